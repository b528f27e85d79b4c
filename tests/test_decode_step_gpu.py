"""The decode-step example: the operators together, in a graph, against the block in 64 bits.

The reference makes every rounding to a stored format that the block makes, but from 64-bit values:
where a value lies next to a rounding boundary the two differ by a unit in the last place.  With an
fp32 error of 2⁻²⁰ that happens to 2⁻²⁰ / 2⁻⁸ of the bf16 values (2⁻¹² of them), each by at most 2⁻⁷;
an e4m3 value by 2⁻³ in 2⁻¹⁶ of them.  In the 2-norm of a row that is 2⁻⁷·2⁻⁶ = 2⁻¹³ for each of three
roundings, and 2⁻³·2⁻⁸ = 2⁻¹¹ for the cache; the bf16 output itself adds 2⁻⁹ at most 2⁻⁸: below 1e-2."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("batch", [1, 5, 16])
def test_decode_step_example(batch, cache):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.main(["--batch", str(batch), "--cache", cache]) < 1e-2
