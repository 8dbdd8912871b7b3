"""GPU parity of a draft step's calls at the edges of what they allow: rows of probabilities that end inside a 16-byte load."""
import numpy as np
import pytest
import torch

import oracle
from attention_attn_fwd_06_gb300 import binding as AB
from attention_attn_fwd_06_gb300.build import build
from tests.test_gpu_drafts import bf16, i32, probabilities

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    AB.load()
    AB.attn_get_device_status()


# ---------------------------------------------------------------- verification of drafts

def padded(x, fill):
    """x [..., V] as a view of rows on 16 bytes, padded past V with `fill`."""
    V = x.shape[-1]
    wide = torch.full((*x.shape[:-1], (V + 8) // 8 * 8), fill, dtype=x.dtype, device=DEV)
    wide[..., :V] = x.to(DEV)
    assert wide.data_ptr() % 16 == 0
    return wide[..., :V]


LAST_NUMBERS = [0.0, 0.3, 1 - 2.0 ** -24, 1.0, float("inf"), float("nan")]


@pytest.mark.parametrize("form", ["drawn", "point", "all", "packed"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 33, 37, 260, 1003, 50257])
def test_verify_drafts_rows_that_end_inside_a_load(V, dtype, form):
    """Padding past the last token would win every draw; the last tokens hold weight; numbers up to 1 and past it."""
    g = np.random.default_rng(V)
    B = len(LAST_NUMBERS)
    q = torch.from_numpy(probabilities(B, V, g)).view(B, 1, V)
    p = torch.from_numpy(probabilities(2 * B, V, g)).view(B, 2, V)
    q[..., -5:], p[..., -5:] = 0.25 * p[:, :1, -5:] + 0.001, p[..., -5:] + 0.002
    p, q = p.to(dtype), q.to(dtype)
    draft = (q - p[:, :1]).float().argmax(-1)  # where the draft's row is furthest above the target's
    u = np.full((B, 2), 1 - 2.0 ** -24, np.float32)
    if form == "all":
        u[:, 0] = 0.0
    u[:, 1] = LAST_NUMBERS
    rows, kw = padded(p, 60000.0), {}
    if form == "packed":
        rows, kw["cu_target"] = rows.flatten(0, 1), i32(2 * np.arange(B + 1))
        assert rows.stride(0) % 8 == 0
    if form != "point":
        kw["draft_probs"] = padded(q, -60000.0)
    tokens, accepted, _ = AB.attn_verify_drafts(i32(draft), rows, torch.from_numpy(u).to(DEV), **kw)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    for b in range(B):
        stand, token = oracle.verify_drafts(draft[b].tolist(), p[b].float().numpy(), u[b].tolist(),
                                            None if form == "point" else q[b].float().numpy())
        assert accepted[b] == stand and tokens[b].tolist() == draft[b, :stand].tolist() + [token] + [-1] * (1 - stand), LAST_NUMBERS[b]
    if form == "all":
        assert (accepted == 1).all()


