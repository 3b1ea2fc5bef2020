"""The example that runs the attention operators and the routed-expert block as one decoder
layer, its step captured and replayed while the sequences grow."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    import __graft_entry__ as g
    g.build()
    import examples.decode_layer as mod
    torch.cuda.set_device(0)
    return mod


@pytest.mark.parametrize("fmt,page,batch,prompt,steps", [("e4m3", 16, 3, 37, 5), ("bf16", 7, 12, 300, 9),
                                                         ("e4m3", 64, 1, 1, 3)])
def test_decode_layer(example, fmt, page, batch, prompt, steps):
    """The attention of the last replayed step against a plain form over the rows read back: its
    weights are rounded to bf16 at most (2^-8) and so is its result (2^-8 of values no larger
    than their mean size); rows read back as bf16 add 2^-8 to each logit's terms (of sizes
    that sum to at most |q| |k| / sqrt(D) < 12 here, doubled for both ends of the softmax) and
    2^-8 to each value."""
    r = example.run(batch=batch, prompt=prompt, steps=steps, fmt=fmt, page=page, check=True)
    # the step before the capture and the replays (a capture runs nothing)
    assert r["lens"] == [prompt + 1 + steps] * batch
    assert torch.isfinite(r["out"]).all()
    back = 0.0 if fmt == "bf16" else 2 * 12 + 1
    assert r["error"] <= (2 + back) * 2.0 ** -8
