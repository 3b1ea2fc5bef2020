"""The example's prompts through prefill, and its steps over a 4-bit cache."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("fmt,page,batch,prompt,steps", [("mxfp4", 16, 3, 37, 5), ("mxfp4", 64, 2, 700, 3), ("bf16", 7, 3, 300, 2),
                                                         ("e4m3", 16, 2, 129, 2)])
def test_prompt_and_steps(fmt, page, batch, prompt, steps):
    """As the example's other test: weights and results rounded to bf16 (2^-8 each); E4M3 rows read back as
    bf16 add 2^-8 to each logit's terms (below 12, doubled) and to each value; MXFP4 rows and bf16 rows are
    bf16 numbers."""
    import __graft_entry__ as g
    g.build()
    import examples.decode_layer as example
    torch.cuda.set_device(0)
    r = example.run(batch=batch, prompt=prompt, steps=steps, fmt=fmt, page=page, check=True)
    assert r["lens"] == [prompt + 1 + steps] * batch and torch.isfinite(r["out"]).all()
    back = 2 * 12 + 1 if fmt == "e4m3" else 0.0
    assert r["error"] <= (2 + back) * 2.0 ** -8 and r["prompt_error"] <= (2 + back) * 2.0 ** -8
