"""What the recurrent block's functions make for a given stream comes from that stream's pool: a block of the current
stream's may still be written there, by work queued before it was freed."""
import pytest
import torch

import gated_linear_recurrence_conv1d_amd as rg
from workloads import WORKLOADS, make_cotangents, make_inputs, to_device

pytestmark = pytest.mark.gpu


def calls():
    inp = make_inputs(WORKLOADS["rg2b"], seed=5, B=2, T=150, D=512, H=2, bias_var=0.25)
    g, ct = to_device(inp, "cuda"), make_cotangents(inp, seed=6)
    par = [g[n] for n in ("conv_w", "W_a", "b_a", "W_x", "b_x", "Lam")]
    dy, dh = torch.from_numpy(ct["dy"]).to("cuda", torch.bfloat16), torch.from_numpy(ct["dh_T"]).cuda()
    y, h = rg.forward(g["x"], *par)
    cs = rg.prefill_state(g["x"])
    q, k = torch.randn(2, 200, 3, 64, device="cuda").bfloat16(), torch.randn(2, 200, 64, device="cuda").bfloat16()
    return [
        ("forward", lambda s: rg.forward(g["x"], *par, stream=s)),
        ("chunked", lambda s: rg.forward(g["x"], *par, plan="chunked", stream=s)),
        ("prefill_state", lambda s: rg.prefill_state(g["x"], stream=s)),
        ("decode_step", lambda s: rg.decode_step(g["x"][:, 0].contiguous(), cs.clone(), h.clone(), *par, stream=s)),
        ("backward", lambda s: rg.backward(g["x"], *par, None, y, dy, dh, stream=s)),
        ("local_mqa", lambda s: rg.local_mqa(q, k, k, 40, stream=s)),
    ]


def test_given_stream_owns_what_is_made_for_it():
    side = torch.cuda.Stream()
    for name, call in calls():
        want = call(None)
        want = list(want.values()) if isinstance(want, dict) else list(want) if isinstance(want, tuple) else [want]
        for given in (side, side.cuda_stream):
            torch.cuda.synchronize()
            got = call(given)
            torch.cuda.synchronize()
            got = list(got.values()) if isinstance(got, dict) else list(got) if isinstance(got, tuple) else [got]
            for a, b in zip(got, want):
                at = a.data_ptr()
                pools = [s["stream"] for s in torch.cuda.memory_snapshot()
                         if s["address"] <= at < s["address"] + s["total_size"]]
                assert pools == [side.cuda_stream], name
                assert torch.equal(a, b), name
