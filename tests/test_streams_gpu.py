"""Calls that are given a stream: what they create belongs to it, whatever the caller's current stream does meanwhile."""
import numpy as np
import pytest
import torch

import cg_tensor_products_b200 as etp
import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _delay(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


def test_results_and_workspaces_of_a_call_on_another_stream():
    """Every call with all but one of its results dropped before its stream has begun, while the current stream
    allocates and fills blocks of the same sizes; and a result dropped while the current stream still reads it."""
    wl = workloads.random_graph(np.random.default_rng(0), 2000, 30000, 2, 16, 15)
    plan = etp.Plan("0..2", 2, "0..2", wl.C)
    t = {k: torch.from_numpy(np.ascontiguousarray(getattr(wl, k))).cuda() for k in ("row_ptr", "src", "r", "x", "w", "g")}
    row_ptr, src, r, x, w, g = (t[k] for k in ("row_ptr", "src", "r", "x", "w", "g"))
    N, E = wl.N, wl.E
    rev = etp.build_reverse_csr(N, row_ptr, src)
    pos = torch.rand(N, 3, device="cuda") * 20
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    W1 = torch.randn(8, 64, generator=gen, device="cuda")
    W2 = torch.randn(64, plan.n_paths * plan.C, generator=gen, device="cuda") / 8
    ggx = torch.randn(x.shape, generator=gen, device="cuda")
    s, here = torch.cuda.Stream(), torch.cuda.current_stream()
    calls = [lambda **k: etp.build_reverse_csr(N, row_ptr, src, **k)[1],
             lambda **k: etp.build_reverse_csr_static(N, row_ptr, src, **k)[0],
             lambda **k: etp.edge_frames(plan, r, **k),
             lambda **k: etp.forward(plan, row_ptr, src, r, x, w, **k),
             lambda **k: etp.backward(plan, row_ptr, src, *rev, r, x, w, g, **k)[1],
             lambda **k: etp.double_backward(plan, row_ptr, src, *rev, r, x, w, g, gg_x=ggx, **k)["grad_w"],
             lambda **k: etp.cart_backward(plan, row_ptr, src, *rev, r, x, w, g, **k)[0],
             lambda **k: etp.radial_forward(plan, r, W1, W2, 5.0, **k),
             lambda **k: etp.fused_forward(plan, row_ptr, src, r, x, W1, W2, 5.0, **k),
             lambda **k: etp.node_product(plan, x, w[:2], **k),
             lambda **k: etp.assemble_forces(N, row_ptr, rev[0], rev[1], r, **k)[0],
             lambda **k: etp.locality_schedule(N, row_ptr, src, pos, 5.0, **k).order]
    for call in calls:
        want = call().clone()
        torch.cuda.synchronize()
        _delay(s)
        got = call(stream=s)
        fill = [torch.full((n,), 1.5e9, device="cuda") for n in (N + 1, E, 3 * N, 3 * E, x.numel(), w.numel(), 88 * E, 1 << 20)
                for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(bool((f == 1.5e9).all()) for f in fill)
        del got, fill
        got = call(stream=s)
        here.wait_stream(s)
        _delay(here)
        later = got.clone()
        del got
        other = call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(later, want) and torch.equal(other, want)
    assert etp.device_fault() == 0


def test_validate_csr_reads_its_flag_on_its_stream():
    row_ptr = torch.tensor([0, 2, 1, 4], dtype=torch.int32, device="cuda")
    src = torch.tensor([0, 1, 7, 2], dtype=torch.int32, device="cuda")
    want = etp.validate_csr(3, row_ptr, src)
    assert want == etp.CSR_NOT_MONOTONE | etp.CSR_SRC_RANGE
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    _delay(s)
    assert etp.validate_csr(3, row_ptr, src, stream=s) == want
