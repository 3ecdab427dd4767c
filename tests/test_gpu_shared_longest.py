"""pa_decode_shared at the longest lengths there are."""
import math

import numpy as np
import pytest
import torch

from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_14_gb300 import build
    B.load(build.build())


@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_FP8])
@pytest.mark.parametrize("back", [0, 1])
def test_the_longest_lengths(kv, back):
    """2^31 - 16 tokens and a block fewer: positions at the end of 32 bits.
    The table names 4096 blocks over and over, whose keys score 0 and whose
    values are 0, and 80 blocks of their own at its end, whose keys score about
    30: e^30 times 1275 keys against 2^31, so all others weigh 2e-7.  The last
    step of 128 keys is a short one, and what lies behind its keys in shared
    memory are keys of the last 80 blocks too, which must not count again."""
    D, nb, cold, hot = 64, (1 << 27) - 1, 4096, 80
    if torch.cuda.mem_get_info()[0] < 4 << 30:
        pytest.skip("4 GB of memory")
    fp8 = kv == W.KV_FP8
    g = torch.Generator().manual_seed(31)
    code = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k = torch.zeros(cold + hot, 1, 16, D)
    v = torch.zeros(cold + hot, 1, 16, D)
    k[cold:, ..., 0] = 7.5 + 0.5 * torch.randint(-2, 3, (hot, 1, 16), generator=g)
    v[cold:] = torch.randint(-8, 9, (hot, 1, 16, D), generator=g) / 4
    table = (torch.arange(nb, dtype=torch.int32, device=DEV) % cold).view(1, nb)
    last = nb - back
    table[0, last - hot:last] = torch.arange(cold, cold + hot, dtype=torch.int32, device=DEV)
    n = last * 16 - 5
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 4
    pools = [(t.to(code).view(torch.uint8) if fp8 else t.to(code)).to(DEV) for t in (k, v)]
    d = B.make_desc(cold + hot, 1, 1, D, B.PA_KV_FP8_E4M3 if fp8 else B.PA_KV_BF16, k_scale=1.0 if fp8 else 0.0,
                    v_scale=1.0 if fp8 else 0.0)
    out, lse = torch.zeros(1, 1, D, device=DEV), torch.zeros(1, 1, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    B.pa_decode_shared(d, out, q, *pools, table, torch.tensor([n], dtype=torch.int32, device=DEV), n,
                       torch.zeros(1, dtype=torch.int32, device=DEV), none, 0, 0, 1.0,
                       B.decode_shared_workspace(d, 1, 0, 0), lse=lse)
    torch.cuda.synchronize()
    s = 4 * k[cold:].to(code).double()[:, 0, :, 0].reshape(-1)[:-5]  # (the bytes' values)
    w = torch.exp(s - 30)
    rest = (n - s.numel()) * math.exp(-30)
    want = (w[:, None] * v[cold:].to(code).double()[:, 0].reshape(-1, D)[:-5]).sum(0) / (w.sum() + rest)
    # exact scores and values, weights good to P's pair (2^-16) and a few 2^-22; |v| <= 2: 1e-4 covers both twice over
    assert np.abs(out[0, 0].double().cpu().numpy() - want.numpy()).max() <= 1e-4
    assert abs(float(lse) - (30 + math.log(float(w.sum()) + rest))) <= 1e-4
