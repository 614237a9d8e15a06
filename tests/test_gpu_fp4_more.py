"""The FP4 stages where their buffers meet: outputs in the place of inputs that have been read, and weights written by
the call just before; and every schedule of the linear."""
import pytest
import torch

import mtp_speculative_draft_head_gb300 as m
import synth
from linear_fp4_schedule import schedule
from test_gpu_fp4 import DEV, EPS, bf16, check_linear, make_copy, rng_matrix

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


# Rows, columns and k, the activation rows a tile, and how the tiles are taken: k split over a cluster, one tile a
# CTA, several (three at least) through two accumulators, or several in groups of activation tiles. On 152 SMs.
SCHEDULES = [
    (9, 60001, 700, 16, "many"),
    (27, 60001, 700, 32, "many"),
    (50, 60001, 700, 64, "many"),
    (90, 3333, 700, 128, "split"),
    (1345, 777, 100, 128, "one"),
    (70, 60001, 700, 128, "many"),
    (225, 20300, 1500, 128, "many"),
    (99, 60001, 2100, 128, "groups"),
    (1345, 777, 1024, 192, "split"),
    (450, 5200, 100, 192, "one"),
    (300, 20300, 700, 192, "many"),
    (140, 60001, 2100, 192, "groups"),
    (193, 5000, 2000, 224, "split"),
    (1000, 3333, 100, 224, "one"),
    (2001, 6200, 1000, 224, "many"),
    (4001, 6200, 700, 224, "many"),
    (201, 30200, 4100, 224, "groups"),
]


@pytest.mark.parametrize("R,N,K,nt,kind", SCHEDULES)
def test_linear_schedules_against_fp64(R, N, K, nt, kind):
    """Every tile width in every way it is run, with ragged last tiles of rows and of weights: sampled rows and
    columns (the first and last of each tile border among them) against 64 bits, the others written."""
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        s = schedule(R, N, K)
        assert s["nt"] == nt and kind == ("split" if s["splits"] > 1 else "groups" if s["group"] else
                                          "one" if s["per_cta"] == 1 else "many")
        assert kind != "many" or s["per_cta"] >= 3
    g = torch.Generator(DEV).manual_seed(R + N)
    x = torch.randn(R, K, device=DEV, generator=g).bfloat16()
    w4, _ = make_copy((torch.randn(N, K, device=DEV, generator=g) * 0.02).bfloat16())
    y = torch.full((R, N), 1e30, dtype=torch.bfloat16, device=DEV)
    m.mtp_head_linear_fp4(x, *w4, y, m.linear_fp4_workspace(R, N, K, DEV))
    rows = {r for t in range(0, R, nt) for r in (t, t + 1, t + nt // 2, t + 127, t + 128, t + nt - 1)} | {R - 1}
    cols = {c for c in range(0, N, max(1, N // 300))} | {c for t in range(0, N, 128 * max(1, N // 12800)) for c in (t, t + 127)}
    cols |= set(range(max(0, N - 140), N))
    rows, cols = (torch.tensor(sorted(i for i in v if i < n), device=DEV) for v, n in ((rows, R), (cols, N)))
    check_linear(x[rows].contiguous(), tuple(t[cols].contiguous() for t in w4), y[rows][:, cols])
    assert not bool((y == 1e30).any())
