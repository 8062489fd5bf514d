"""Calls that take several launches or more LDS than a launch has unasked, captured
into a HIP graph and replayed with eager calls between: prompts of the scan that are
cut into chunks, and the norm's gradients over many tokens of wide groups."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

from test_gpu_scan import device_args, inputs

pytestmark = pytest.mark.gpu


def replayed(run, fill, n=4):
    """``run()`` captured once; every replay on contents ``fill(k)`` against an eager run."""
    want = []
    for k in range(2):
        fill(k)
        want.append([t.clone() for t in run()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for turn in range(n):
        fill(turn % 2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[turn % 2]):
            assert torch.equal(a, b), f"replay {turn}"
        fill(1 - turn % 2)
        run()
        torch.cuda.synchronize()


@pytest.mark.parametrize("N", [8, 16, 64])
def test_a_prompt_cut_into_chunks(N):
    case = (2, 1100, 24, N, 2, "bf16", True, True, True, True, True, [1100, 905], False)
    sets = [device_args(*inputs(case, seed=s)) for s in (81, 82)]
    main = [t.clone() for t in sets[0][0]]
    a = {k: v.clone() if torch.is_tensor(v) else v for k, v in sets[0][1].items()}

    def fill(k):
        for t, v in zip(main, sets[k][0]):
            t.copy_(v)
        for name, v in sets[k][1].items():
            if torch.is_tensor(v):
                a[name].copy_(v)

    replayed(lambda: fb.falcon_scan_fwd(*main, **a), fill)


def test_gradients_of_a_norm_of_wide_groups_over_many_tokens():
    tokens, G, d = (1 << 15) + 77, 4, 2048          # more than 64 tokens a thread, 64 KiB of LDS for their sums
    x = torch.empty(1, tokens, G * d, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty(1, tokens, G * d, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(G * d, device="cuda")

    def fill(k):
        g = torch.Generator(device="cuda").manual_seed(90 + k)
        x.normal_(generator=g)
        dy.normal_(generator=g)

    def run():
        g = fb.falcon_norm_bwd(x, G, dy, w, w, activation="silu", center=True)
        return g["dweight"], g["dbias"], g["dx"]

    replayed(run, fill, n=2)
    torch.cuda.empty_cache()
