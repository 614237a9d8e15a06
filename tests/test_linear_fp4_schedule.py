"""The FP4 linear's choice of schedule over its whole range, without a GPU: what the kernels take for granted."""
import random

import pytest

from linear_fp4_schedule import schedule
from test_gpu_fp4_more import SCHEDULES


@pytest.mark.parametrize("sms", [152, 148, 8])
def test_every_shape_has_a_schedule_that_its_workspace_and_cluster_hold(sms):
    rng = random.Random(sms)
    shapes = [(r, n, k) for r in (1, 128, 129, 65536) for n in (1, 128, 2 ** 31 - 1) for k in (1, 256, 131072)]
    shapes += [tuple(int(2 ** rng.uniform(0, b)) for b in (16, 22, 17)) for _ in range(3000)]
    for R, N, K in shapes:
        if (R + 15) // 16 * ((N + 127) // 128) >= 2 ** 31:
            continue  # (y would be beyond any memory)
        s = schedule(R, N, K, sms)
        assert s["nt"] in (16, 32, 64, 128, 192, 224) and 1 <= s["splits"] <= 8, (R, N, K)
        assert s["mt"] == -(-N // 128) and s["tiles"] == s["mt"] * -(-R // s["nt"])
        # whole 128-row scale blocks per activation tile, in a workspace that counts 8, or R / 64 + 2 of them
        blocks = -(-R // s["nt"]) * -(-s["nt"] // 128)
        assert blocks <= (8 if R <= 128 else -(-R // 64) + 2), (R, N, K)
        if s["splits"] > 1:
            # all clusters at once, a stage at least for each CTA, and the partial sums fit the first one's ring
            assert s["tiles"] * s["splits"] <= sms and s["splits"] <= s["nkb"]
            assert (s["splits"] - 1) * s["nt"] * 128 * 4 <= 160 * 1024 and not s["group"]
        if s["group"]:
            assert s["nt"] >= 128 and s["tiles"] >= sms


def test_the_gpu_tests_reach_every_schedule():
    seen = {(nt, kind) for _, _, _, nt, kind in SCHEDULES}
    for nt in (128, 192, 224):
        assert {(nt, k) for k in ("split", "one", "many", "groups")} <= seen
    assert {(nt, "many") for nt in (16, 32, 64)} <= seen
