"""Loads of the non-coherent path are for memory that nothing writes while a kernel runs.  Kernels start before the one
before them has ended, so what that one may write (activations, logits, settings) is loaded otherwise."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bloom_decoder_token_gb300", "csrc")
# A model's weights, which no kernel writes: a layer norm's, fused into the linear layer; a linear layer's.
CONSTANT = {"__ldg(reinterpret_cast<const uint2 *>(a.ln_g + k))", "__ldg(reinterpret_cast<const uint2 *>(a.ln_b + k))",
            "ld_stream(wp[r] + (size_t)c * KC * (INT8 ? 1 : 2))"}


def code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def test_non_coherent_loads_are_of_weights():
    seen = set()
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = code(path)
        assert "__restrict__" not in text, path      # with it the compiler may choose such loads by itself
        for m in re.finditer(r"\b(__ldg|ld_stream)\(", text):
            if text[: m.start()].endswith("__forceinline__ uint4 "):
                continue                             # the helper's own definition
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            call = re.sub(r"\s+", " ", text[m.start(): end])
            assert call in CONSTANT, (os.path.basename(path), call)
            seen.add(call)
        assert len(re.findall(r"\.nc\b", text)) == (1 if path.endswith("common.cuh") else 0), path   # ld_stream's
    assert seen == CONSTANT
