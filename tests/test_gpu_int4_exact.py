"""INT4 products whose every float32 step is exact: activations -3 .. 3, scales that are
powers of two from 1/8 to 1, so that one code, scale, zero point or value out of place
changes a result.  A product with 16 + q is at most 93 and a group's sum below 2^14; a
whole sum is at most 8224 products of 45 in steps of 1/8, below 2^22 of them: every order
of additions gives the same float32."""
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu

F = {"bf16": torch.bfloat16, "f16": torch.float16}

# E, N, rows of each expert in turn; reductions above 512 unless said
TASKS = {
    "one_tile": (1, 96, [3]),                             # one tile a wave: fewer workgroups than CUs
    "one_tile_experts": (5, 40, [1, 0, 17, 2, 16]),
    "two_tiles": (8, 1040, [1, 2, 0, 5, 1, 16, 33, 3]),   # 33 column groups of 32 an expert
    "four_tiles": (16, 1040, [1, 2, 0, 5, 1, 16, 33, 3] * 2),
}
LONG = [32 * 17, 32 * 33, 32 * 37, 32 * 65, 32 * 193, 32 * 257]    # rounded up to whole groups
SHORT_TASKS = {
    "few_rows": (3, 100, [1, 16, 7]),
    "rounds": (128, 8200, [2] * 128),                     # several column groups a wave
    "many_rows": (3, 100, [33, 0, 17]),                   # two row tiles a wave
    "many_rows_rounds": (64, 8200, [40] * 64),
}


def _product(E, N, K, rows, group, zeros, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def ints(lo, hi, shape, t):
        return torch.randint(lo, hi, shape, generator=g, device=DEV).to(t)

    off = torch.tensor([0] + rows, device=DEV).cumsum(0).to(torch.int32)
    M = sum(rows)
    x = ints(-3, 4, (M, K), F[dtype])
    codes = ints(0, 256, (E, N, K // 2), torch.uint8)
    scales = 2.0 ** ints(-3, 1, (E, N, K // group), torch.float32)
    z = ints(0, 16, scales.shape, torch.uint8) if zeros else None
    got = m.int4_grouped_gemv(x, m.INT4Tensor(codes, scales.to(F[dtype]), z, group), off, m_total=M, out_dtype=torch.float32)
    at = 0
    for e, n in enumerate(rows):
        if n == 0:
            continue
        q = torch.stack([codes[e] & 15, codes[e] >> 4], -1).view(N, K // group, group).double()
        q -= 8.0 if z is None else z[e].double()[..., None]
        b = (q * scales[e].double()[..., None]).view(N, K)
        want = x[at:at + n].double() @ b.T
        assert torch.equal(got[at:at + n].double(), want), (e, torch.nonzero(got[at:at + n].double() != want)[:5])
        at += n
    # rounded to 16 bits once
    low = m.int4_grouped_gemv(x, m.INT4Tensor(codes, scales.to(F[dtype]), z, group), off, m_total=M)
    finite = got.abs() < 65504
    assert torch.equal(low[finite], got.to(F[dtype])[finite])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("task", TASKS)
def test_long_reductions(task, group, zeros, dtype):
    E, N, rows = TASKS[task]
    for K in LONG:
        K = (K + group - 1) // group * group
        print("exact", task, K, group, zeros, dtype, flush=True)
        _product(E, N, K, rows, group, zeros, dtype, K)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("task", SHORT_TASKS)
def test_short_reductions(task, group, zeros, dtype):
    E, N, rows = SHORT_TASKS[task]
    for K in sorted({(k + group - 1) // group * group for k in ([32, 160, 512] if N > 1000 else [32, 96, 160, 256, 288, 416, 512])}):
        print("exact", task, K, group, zeros, dtype, flush=True)
        _product(E, N, K, rows, group, zeros, dtype, K)
