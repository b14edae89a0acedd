"""Rotation and norms over more tokens than one launch takes: each stretch as a call on it alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

puro = pytest.importorskip("blockwise_fp8_gemm_act_amd")

TOKENS = (1 << 26) + 5
STRETCHES = [slice(0, 9), slice((1 << 25) - 5, (1 << 25) + 5), slice((1 << 26) - 5, TOKENS)]


@pytest.fixture(scope="module")
def data():
    """One head of 64 for each token: short random rows repeated, so that making them takes no time."""
    g = torch.Generator(device="cuda").manual_seed(1)
    row = torch.randn(1021, 64, generator=g, device="cuda").to(torch.bfloat16)
    x = row.repeat(-(-TOKENS // 1021), 1)[:TOKENS]
    pos = torch.randint(0, 100, (TOKENS,), generator=g, device="cuda", dtype=torch.int32)
    yield x, pos, puro.rope_table(100, 64)
    torch.cuda.empty_cache()


def test_rope(data):
    x, pos, table = data
    y = puro.rope(x[:, None], table, pos)
    for s in STRETCHES:
        assert torch.equal(y[s], puro.rope(x[s, None], table, pos[s].clone()))
    plain = puro.rope(x[:, None], table)                 # no positions given: a token's own number
    assert torch.equal(plain[:100], puro.rope(x[:100, None], table)) and bool(plain[100:1000].isnan().all())
    assert bool(plain[STRETCHES[1]].isnan().all()) and bool(plain[STRETCHES[2]].isnan().all())


def test_norm_and_rotation(data):
    x, pos, table = data
    w = torch.linspace(0.5, 1.5, 64, device="cuda").to(torch.bfloat16)
    q, _ = puro.qk_norm_rope(x, w, w, table, pos, q_heads=1, k_heads=0)
    for s in STRETCHES:
        assert torch.equal(q[s], puro.qk_norm_rope(x[s], w, w, table, pos[s].clone(), q_heads=1, k_heads=0)[0])
