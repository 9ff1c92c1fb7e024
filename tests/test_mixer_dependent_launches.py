"""Kernels of the operators around the token mixers that launch_pdl starts while the kernel before them runs:
each waits for the stream before anything that may read or write global memory.  On the sources; no GPU."""
import os
import re

import pytest

import linear_attention_attn_b200 as la

CSRC = os.path.join(os.path.dirname(la.__file__), "csrc")
SOURCES = ("la_conv.cu", "la_norm.cu", "la_scan.cu", "la_scan_bwd.cu")
ACCESS = re.compile(r"\bload_\w+\s*[<(]|\bstore_\w+\s*[<(]|\.load\(|\.store\(|\bldv<|\bstv<|\b(?:a|sg)\.\w+\[|\bpart\[|\bchan\[")


def _launched():
    for name in SOURCES:
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for kernel in sorted(set(re.findall(r'launch_pdl\(\s*"\w+",\s*(\w+)', text))):
            yield name, kernel, text


@pytest.mark.parametrize("name,kernel", [(n, k) for n, k, _ in _launched()])
def test_waits_before_its_first_access(name, kernel):
    text = next(t for n, k, t in _launched() if (n, k) == (name, kernel))
    body = text[text.index("{", re.search(r"\b%s\(" % kernel, text).start()):]
    before = body[:body.index("wait_for_stream()")]
    assert "\n}\n" not in before, "no wait in this kernel"
    found = ACCESS.search(before)
    assert not found, "%r before the wait" % found.group(0)


def test_the_kernels_are_found():
    assert {k for _, k, _ in _launched()} == {"conv_bwd_reduce", "norm_join", "norm_apply", "norm_bwd_apply",
                                              "scan_fwd_kernel", "scan_bwd_kernel", "scan_bwd_join"}
