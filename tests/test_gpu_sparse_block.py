"""The example that runs the projection with adapters, the router and the experts
together: prompt tokens, then decoding from a CUDA graph, against 64 bits (it
returns the worst row's distance in the 2-norm; three bf16 roundings of about
0.42 * 2^-8 each, and int8 codes that fp32 sums move by one, stay inside 1e-2)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("variant", ["w4a8", "w4a16"])
@pytest.mark.parametrize("tokens,requests", [(1, 1), (77, 5), (700, 33)])
def test_sparse_block(variant, tokens, requests):
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "sparse_block.py")
    spec = importlib.util.spec_from_file_location("sparse_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors = example.main(["--tokens", str(tokens), "--requests", str(requests), "--hidden", "512",
                           "--inner", "256", "--experts", "16", "--picks", "4", "--adapters", "6",
                           "--rank", "16", "--variant", variant])
    assert max(errors) < 1e-2
