"""The operators around a student's blocks on the GPU where test_gpu_ops_block does not reach:
arrays that lie between one another, the ends of binary32, long sums of one sign."""
import math

import pytest

import ops_block_ref as B
import ops_ref as R
from gpu_util import gpu_or_skip
from test_gpu_ops_block import _gen, _rand, _same, _types, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zs():
    gpu_or_skip()
    import zero_sharded_mixed_step_amd as zs
    zs.ops_lib()
    return zs


@pytest.fixture(scope="module")
def torch():
    return gpu_or_skip()


@pytest.mark.parametrize("T,C", [(1, 64), (37, 64), (300, 1000)])
def test_columns_of_one_buffer(zs, torch, T, C):
    """Inputs and outputs that are columns of one buffer, or its rows in turn, are apart: the same
    bits as in buffers of their own."""
    bf = torch.bfloat16
    g = _gen(torch, T)
    x, y, dh, dz, d = (_rand(torch, g, (T, C), bf).cuda() for _ in range(5))
    w = _rand(torch, g, (C,), bf, 0.3).cuda()
    ids = torch.randint(-1, T, (T,), generator=g, dtype=torch.int32).cuda()
    kw = dict(post_norm=True, post_weight=w, gate=w, pre_weight=w)
    ws = _ws(torch, max(zs.zero_block_norm_workspace_bytes(T, C), zs.zero_embed_workspace_bytes(T, C)))[0]

    def run(x, y, dh, dz, d, h, z, dx, dy, dt):
        zs.zero_block_norm_fwd(x, y, h, z, **kw)
        zs.zero_block_norm_bwd(y, h, dh, dz, dx, dy, **kw)
        zs.zero_embed_bwd(ids, d, dt, workspace=ws)
        return h, z, dx, dy, dt

    want = run(x, y, dh, dz, d, *(torch.empty_like(x) for _ in range(5)))
    columns = torch.full((T, 10 * C), math.nan, dtype=bf, device="cuda").view(T, 10, C).unbind(1)
    turns = torch.full((T, 10, C), math.nan, dtype=bf, device="cuda").unbind(1)
    for v in (columns, turns):
        for to, of in zip(v, (x, y, dh, dz, d)):
            to.copy_(of)
        for a, b in zip(run(*v), want):
            assert _same(a, b)
