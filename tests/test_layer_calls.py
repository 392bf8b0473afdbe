"""The calls that ``run_layer`` makes, in their order, with the library's entry points
replaced by a record of their names."""
import pytest
import torch

B = pytest.importorskip("mixture_experts_layer_plan_amd.binding")

ENTRIES = ("moe_route", "moe_plan", "moe_quantize_weights_mxfp8", "moe_forward_mxfp8", "moe_backward_mxfp8",
           "moe_forward_bf16", "moe_backward_bf16", "moe_route_backward", "moe_adamw_table", "moe_adamw_step",
           "moe_lora_plan", "moe_lora_bf16", "moe_lora_backward_bf16")
SHORT = {"moe_quantize_weights_mxfp8": "quantise", "moe_forward_mxfp8": "forward", "moe_forward_bf16": "forward",
         "moe_adamw_step": "step"}


@pytest.fixture
def calls(monkeypatch):
    got = []
    for name in ENTRIES:
        monkeypatch.setattr(B, name, lambda *a, name=name: got.append(SHORT.get(name)))

    def take():
        out = [n for n in got if n]
        got.clear()
        return out
    return take


def layer(dtype):
    from mixture_experts_layer_plan_amd import AdamW, LayerBuffers
    T, H, I, E, k = 4, 128, 128, 2, 1
    b = LayerBuffers(T, H, I, E, k, dtype=dtype, device="cpu")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)    # noqa: E731
    inp = dict(x=z(T, H), logits=torch.zeros(T, E), w_gate=z(E, I, H), w_up=z(E, I, H), w_down=z(E, H, I),
               dy=z(T, H))
    return b, inp, AdamW(b, inp, 8), B.adamw_hyper(1e-3, seed=1)


def test_no_forward_reads_quantised_weights_from_before_a_step(calls):
    """Whatever ``quantize`` says, a forward behind a step reads the step's weights."""
    from mixture_experts_layer_plan_amd import layer as layer_, run_layer
    b, inp, opt, h = layer("mxfp8")
    calls()
    run_layer(b, inp)
    assert calls() == ["quantise", "forward"]
    run_layer(b, inp, quantize=False)                       # nothing has changed
    assert calls() == ["forward"]
    for _ in range(2):                                      # the same calls again, as a replay makes them
        run_layer(b, inp, quantize=False, adamw=opt, hyper=h)
        assert calls() == ["forward", "step", "quantise"]
    run_layer(b, inp, quantize=False)
    assert calls() == ["forward"]
    for _ in range(2):
        run_layer(b, inp, adamw=opt, hyper=h)
        assert calls() == ["quantise", "forward", "step"]
    run_layer(b, inp, backward=False, quantize=False)
    run_layer(b, inp, quantize=False)
    assert calls() == ["quantise", "forward", "forward"]
    opt.step(h)                                             # a step by itself
    layer_.run_forward(b, inp, quantize=False)
    layer_.run_forward(b, inp, quantize=False)
    assert calls() == ["step", "quantise", "forward", "forward"]
    opt.step(h)
    layer_.quantize_weights(b, inp)                         # and weights quantised by the caller
    layer_.run_forward(b, inp, quantize=False)
    assert calls() == ["step", "quantise", "forward"]


def test_a_bf16_layer_quantises_nothing(calls):
    from mixture_experts_layer_plan_amd import run_layer
    b, inp, opt, h = layer("bf16")
    calls()
    run_layer(b, inp, quantize=False, adamw=opt, hyper=h)
    run_layer(b, inp, quantize=False)
    assert calls() == ["forward", "step", "forward"]


def test_a_step_over_other_weights_or_gradients_is_refused(calls):
    """It would update weights that the forward did not read, or from gradients that the
    backward did not write."""
    from mixture_experts_layer_plan_amd import run_layer
    b, inp, opt, h = layer("bf16")
    b2, inp2, _, _ = layer("bf16")
    for bb, ii in ((b2, inp), (b, inp2), (b, dict(inp, w_up=inp2["w_up"])),
                   (b, {k: v for k, v in inp.items() if k != "w_down"})):
        calls()
        with pytest.raises(ValueError):
            run_layer(bb, ii, adamw=opt, hyper=h)
        assert calls() == []
    run_layer(b, dict(inp, x=inp2["x"], dy=inp2["dy"]), adamw=opt, hyper=h)     # another batch
    assert calls() == ["forward", "step"]
    # buffers for another number of tokens that share the gradients
    for g in ("dw_gate", "dw_up", "dw_down"):
        setattr(b2, g, getattr(b, g))
    run_layer(b2, dict(inp2, **{w: inp[w] for w in ("w_gate", "w_up", "w_down")}), adamw=opt, hyper=h)
    assert calls() == ["forward", "step"]


def test_a_step_over_some_of_the_weights(calls):
    """Weights that the table leaves out stay as they are: an MXFP8 layer's experts too."""
    from mixture_experts_layer_plan_amd import AdamW, LayerBuffers, run_layer
    _, inp, _, h = layer("mxfp8")
    b = LayerBuffers(4, 128, 128, 2, 1, dtype="mxfp8", device="cpu", adapters=(1, 16))
    inp.update(lora_a=torch.zeros(1, 16, 128, dtype=torch.bfloat16),
               lora_b=torch.zeros(1, 128, 16, dtype=torch.bfloat16), lora_scale=torch.zeros(1),
               adapter_idx=torch.zeros(4, dtype=torch.int32))
    opt = AdamW(b, {k: inp[k] for k in ("lora_a", "lora_b")})
    calls()
    run_layer(b, inp, quantize=False, adamw=opt, hyper=h)
    run_layer(b, inp, quantize=False)
    assert calls() == ["forward", "step", "forward"]
