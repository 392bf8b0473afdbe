"""The AdamW step over an MXFP8 layer, whose forward reads quantised copies of the weights:
bit for bit the layer that quantises in every call."""
import pytest
import torch

from gpu_util import digest, say, to_dev
from test_gpu_step_layer import buffers, inputs

pytestmark = pytest.mark.gpu
T = 96
NAMES = ("y", "dx", "loss", "d_logits", "dw_gate", "dw_down")


def start(bits=8):
    from mixture_experts_layer_plan_amd import AdamW, layer
    inp = to_dev(inputs(T, "mxfp8", seed=11))
    b = buffers(T, "mxfp8")
    opt = AdamW(b, inp, bits)
    layer.quantize_weights(b, inp)
    return b, inp, opt


def state(b, inp, opt):
    torch.cuda.synchronize()
    return digest(*[getattr(b, n) for n in NAMES], *[inp[n] for n in opt.state],
                  *[v for st in opt.state.values() for v in st.values()])


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_without_quantising_by_the_caller(bits):
    say(f"AdamW over mxfp8, quantize=False, bits={bits}")
    from mixture_experts_layer_plan_amd import binding as B, run_layer
    runs = []
    for quantize in (True, False):
        b, inp, opt = start(bits)
        got = []
        for step in (1, 2, 3):
            run_layer(b, inp, quantize=quantize, adamw=opt, hyper=B.adamw_hyper(1e-2, step=step, seed=step))
            got.append(state(b, inp, opt))
        runs.append(got)
    assert runs[0] == runs[1] and len(set(runs[0])) == 3


def test_a_forward_behind_a_step_reads_its_weights():
    say("AdamW over mxfp8, forward behind a step")
    from mixture_experts_layer_plan_amd import binding as B, layer, run_layer
    b, inp, opt = start()
    run_layer(b, inp, quantize=False)
    first = b.y.clone()
    opt.step(B.adamw_hyper(1e-1, step=1, seed=1))
    layer.run_forward(b, inp, quantize=False)
    got = b.y.clone()
    layer.run_forward(b, inp)
    torch.cuda.synchronize()
    assert torch.equal(b.y, got) and not torch.equal(first, got)


def test_a_captured_call_with_a_step():
    """Each replay reads the weights that the replay before it left."""
    say("AdamW over mxfp8 in a graph, quantize=False")
    from mixture_experts_layer_plan_amd import binding as B, run_layer
    runs = []

    def put(t, h):
        t.copy_(torch.frombuffer(bytearray(bytes(h)), dtype=torch.uint8))
    for graph in (False, True):
        b, inp, opt = start()
        begin = {k: v.clone() for k, v in inp.items()}
        hd = torch.zeros(40, dtype=torch.uint8, device="cuda")
        put(hd, B.adamw_hyper(1e-2, step=1, seed=1))
        if graph:
            run_layer(b, inp, quantize=False, adamw=opt, hyper=hd)   # the side stream exists
            torch.cuda.synchronize()
            for k, v in begin.items():
                inp[k].copy_(v)
            for st in opt.state.values():
                for v in st.values():
                    v.zero_()
            b.wq.copy_(start()[0].wq)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run_layer(b, inp, quantize=False, adamw=opt, hyper=hd)
        got = []
        for step in (1, 2, 3):
            put(hd, B.adamw_hyper(1e-2, step=step, seed=step))
            if graph:
                g.replay()
            else:
                run_layer(b, inp, quantize=False, adamw=opt, hyper=hd)
            got.append(state(b, inp, opt))
        runs.append(got)
    assert runs[0] == runs[1] and len(set(runs[0])) == 3
