"""attn_fwd_prefix over long own caches and prefixes: the numerics contract (99.9% of outputs
within one unit in the last place) where a part of the keys is tens of thousands long."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

from _parity import assert_parity, bits_of, compare

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


@pytest.mark.parametrize("Hq,Hkv,cap,Sp", [
    (304, 304, 131072, 0),         # two blocks an SM: each cache is one part
    (24 * 304, 304, 131072, 0),    # 24 rows a block
    (10 * 304, 304, 40000, 0),     # 10 rows
    (32 * 304, 304, 20000, 0),     # 32 rows
    (160, 8, 64, 1_200_000),       # a long prefix and few rows
    (30, 1, 64, 1_200_000),        # all parts that the join takes, 18750 keys each
    (2432, 304, 16385, 0),
])
def test_long_parts_keep_the_contract(Hq, Hkv, cap, Sp):
    g = torch.Generator(device="cuda").manual_seed(Hq + cap)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v = r(1, Hq, 1, 128), r(1, Hkv, cap, 128), r(1, Hkv, cap, 128)
    kp, vp = (r(Hkv, Sp, 128), r(Hkv, Sp, 128)) if Sp else (None, None)
    n = torch.tensor([cap], dtype=torch.int32, device="cuda")
    out, lse = attn.attn_fwd_prefix(q, kp, vp, k, v, n)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    want = torch.empty(Hq, 128, dtype=torch.float64)
    group = Hq // Hkv
    for h in range(Hkv):
        rows = slice(h * group, (h + 1) * group)
        keys, vals = k[0, h], v[0, h]
        if Sp:
            keys, vals = torch.cat([kp[h], keys]), torch.cat([vp[h], vals])
        s = q[0, rows, 0].double() @ keys.double().T * SCALE
        assert (lse[0, rows, 0].double() - torch.logsumexp(s, 1)).abs().max() <= 1e-4
        want[rows] = (torch.softmax(s, 1) @ vals.double()).cpu()
    assert_parity(compare(bits_of(out[0, :, 0]), want.numpy(), "rtne"), excess=True)
