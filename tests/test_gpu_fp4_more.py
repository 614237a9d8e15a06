"""The FP4 stages where their buffers meet: outputs in the place of inputs that have been read, and weights written by
the call just before."""
import pytest
import torch

import mtp_speculative_draft_head_gb300 as m
import synth
from test_gpu_fp4 import DEV, EPS, bf16, make_copy, rng_matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,N", [(3, 512), (40, 1024), (300, 6144)])
def test_linear_output_in_the_place_of_its_input(R, N):
    x = bf16(rng_matrix(R, N, R) * 50.0)
    w4, _ = make_copy((torch.randn(N, N, device=DEV, generator=torch.Generator(DEV).manual_seed(R)) * 0.02).bfloat16())
    ws = m.linear_fp4_workspace(R, N, N, DEV)
    want = torch.zeros_like(x)
    m.mtp_head_linear_fp4(x, *w4, want, ws)
    y = x.clone()
    m.mtp_head_linear_fp4(y, *w4, y, ws)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("R,H", [(2, 256), (200, 512)])
def test_context_rows_in_the_place_of_target_hidden(R, H):
    V = 400
    g = {k: v.to(DEV) for k, v in synth.make_weights(H, V, 3, "cpu").as_dict().items()}
    tokens, hidden = (t.to(DEV) for t in synth.make_step_inputs(H, V, R, 4, "cpu", distinct=False))
    eh, _ = make_copy(g["eh_proj"])
    ws = m.context_fp4_workspace(R, H, DEV)

    def rows(h, out):
        m.mtp_head_context_rows_fp4(g["embed"], g["enorm_w"], g["hnorm_w"], *eh, tokens, h, out, ws, eps=EPS)
        return out
    want = rows(hidden, torch.zeros_like(hidden))
    both = hidden.clone()
    assert torch.equal(rows(both, both).view(torch.int16), want.view(torch.int16))


def test_dequantised_weights_are_swept_at_once():
    """lm_head written back from its copy and swept by the next call, which streams it from its first cycle on: the
    logits of the weights just written, not of the ones before."""
    H, V, B = 1024, 40000, 3
    gen = torch.Generator(DEV).manual_seed(1)
    copies = [make_copy((torch.randn(V, H, device=DEV, generator=gen) * 0.02).bfloat16())[0] for _ in range(2)]
    x = torch.randn(B, H, device=DEV, generator=gen).bfloat16()
    fw = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    w = torch.empty(V, H, dtype=torch.bfloat16, device=DEV)
    ws = m.workspace(B, H, V, DEV)

    def step(i, b, wait):
        lg, d = torch.zeros(b, V, device=DEV), torch.zeros(b, dtype=torch.int32, device=DEV)
        m.mtp_head_dequantize_fp4(*copies[i], w)
        wait()
        m.mtp_head_logits_argmax_batched(x[:b], fw, w, None, m.W_BF16, lg, d, ws, eps=EPS)
        return lg, d
    for b in (1, B):
        want = [step(i, b, torch.cuda.synchronize) for i in range(2)]
        got = [step(i % 2, b, lambda: None) for i in range(20)]
        for i, (lg, d) in enumerate(got):
            assert torch.equal(lg, want[i % 2][0]) and torch.equal(d, want[i % 2][1])
