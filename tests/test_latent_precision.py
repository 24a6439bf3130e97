"""How many bits the expanded form's values and probabilities keep: a bound that
f16 for both meets and bf16 for either does not.

Scores come from the rotary part alone, which is neither expanded nor rounded,
so keys add no error.  What is left, with u16 = 2^-11 and u = 2^-8 the unit
roundoffs of f16 and bf16: the values u16 sum p|v|, the probabilities as much
again, fp32 sums and scores 2^-12 sum p|v|, the output u |ref|.  The queries see
1 to 64 tokens, so their outputs are far smaller than sum p|v| in many places,
and a bf16 rounding of one operand (2^-8 of each term) stands out."""
import math

import pytest
import torch

import edge_moe_serving_gb300 as moe
from kv_helpers import attend64

U, U16 = 2.0 ** -8, 2.0 ** -11
N, HEADS, RANK, ROPE, DN, DV = 64, 8, 256, 32, 64, 128
SCALE = 0.25


def inputs():
    g = torch.Generator().manual_seed(7)
    rows = torch.randn(N, RANK + ROPE, generator=g).to(torch.bfloat16)
    q = torch.randn(N, HEADS, DN + ROPE, generator=g).to(torch.bfloat16)
    q[:, :, :DN] = 0
    w = (torch.randn(HEADS, DN + DV, RANK, generator=g) / math.sqrt(RANK)).to(torch.bfloat16)
    return rows, q, w


def outside(out, rows, q, w):
    """Places of out [N, HEADS, DV] that are further from the definition than the bound."""
    x, n = rows.double(), 0
    for h in range(HEADS):
        v = x[:, :RANK] @ w[h, DN:].double().T
        ref, mag, _ = attend64(q[:, h, DN:].double(), x[:, RANK:], v, SCALE, list(range(1, N + 1)))
        n += int(((out[:, h].double() - ref).abs() > U * ref.abs() + (2 * U16 + 2.0 ** -12) * mag).sum())
    return n


@pytest.mark.parametrize("p_type,v_type,fits", [(torch.float16, torch.float16, True), (torch.bfloat16, torch.float16, False),
                                                (torch.float16, torch.bfloat16, False), (torch.float32, torch.float32, True)])
def test_the_bound_tells_the_types_apart(p_type, v_type, fits):
    """A plain form with its operands rounded to a type, in place of the kernel."""
    rows, q, w = inputs()
    out = torch.empty(N, HEADS, DV)
    t = torch.arange(N)
    for h in range(HEADS):
        v = (rows[:, :RANK].float() @ w[h, DN:].float().T).to(v_type).float()
        z = (q[:, h, DN:].float() @ rows[:, RANK:].float().T) * SCALE
        z[t[None] > t[:, None]] = -math.inf
        p = torch.exp(z - z.amax(1, keepdim=True)) * 128
        out[:, h] = (p.to(p_type).float() @ v) / p.sum(1, keepdim=True)
    n = outside(out.to(torch.bfloat16), rows, q, w)
    assert (n == 0) == fits, n


@pytest.mark.gpu
def test_the_kernel_is_inside_the_bound():
    from kv_helpers import DEV, Paged

    rows, q, w = inputs()
    c = Paged(N // 32, 32, RANK, ROPE, 1, N // 32)
    c.pages[0] = rows.view(N // 32, 32, -1).to(DEV)
    c.table[0] = torch.arange(N // 32, dtype=torch.int32)
    c.lens[0] = N
    n = moe.moe_latent_prefill_workspace_size(c.handle, 1, N, HEADS, DN, DV, N)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = torch.empty(N, HEADS, DV, dtype=torch.bfloat16, device=DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    moe.moe_latent_prefill(c.handle, 0, q.to(DEV), i32([0]), i32([0, N]), 1, N, HEADS, DN, DV, w.to(DEV), SCALE, N, out,
                           ws, n, c.status)
    assert c.bits() == 0
    assert outside(out.cpu(), rows, q, w) == 0
