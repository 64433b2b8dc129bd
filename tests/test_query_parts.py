"""How the chunk attention over the 8-bit caches holds its queries where rows share
reads: each head row as two E4M3 parts and a power of two. What the header says of
their precision, against every bf16 value beside every largest one (on the host)."""

import os
import re

import torch

import paged_gqa_decode_reshape_gb300 as pg

E4M3 = torch.float8_e4m3fn


def parts(x, largest):
    """What the two parts of bf16 values stand for in a row with this largest magnitude, in fp64."""
    k = (torch.floor(torch.log2(largest)) - 7).clamp(min=-119)  # largest / 2^k in [128, 256)
    y = x * torch.exp2(-k)
    hi = y.float().to(E4M3).double()
    return (hi + (y - hi).float().to(E4M3).double()) * torch.exp2(k)


def stated():
    """The two exponents of the header: values from 2^-a of the largest on are exact, others off by at most 2^-b of it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(pg.__file__)))
    with open(os.path.join(root, "include", "paged_decode.h")) as f:
        text = re.sub(r"\s*\n \* ", " ", f.read())
    a, b = re.search(r"exact for values of at least 2\^-(\d+) of the row's largest, the others off by at most 2\^-(\d+) of it",
                     text).groups()
    return int(a), int(b)


def test_what_the_header_says_of_the_queries():
    a, b = stated()
    m = (128 + torch.arange(128)).double()  # mantissas
    largest = m[:, None, None] / 128
    x = m[None, :, None] / 128 * torch.exp2(-torch.arange(30).double())[None, None, :]
    inside = x <= largest
    off = ((parts(x, largest) - x).abs() / largest)[inside]
    near = (x / largest)[inside]
    assert (off[near >= 2.0 ** -a] == 0).all(), f"not exact up to {near[off > 0].max().item():.3e} of the largest"
    assert off.max() <= 2.0 ** -b, f"off by up to 2^{torch.log2(off.max()).item():.2f} of the largest"
    # and no tighter power of two holds
    assert (off[near >= 2.0 ** -(a + 1)] > 0).any() and off.max() > 2.0 ** -(b + 1)


def test_rows_of_tiny_queries():
    """A row's largest value below 2^-112, down to the smallest bf16 number, counts as 2^-112."""
    a, b = stated()
    x = torch.arange(1, 1 << 12, 3).to(torch.int16).view(torch.bfloat16).double()  # 2^-133 to 2^-95
    for at in range(0, len(x), 7):
        row = x[:at + 1]
        off, largest = (parts(row, row[-1]) - row).abs(), max(row[-1].item(), 2.0 ** -112)
        assert off.max() <= 2.0 ** -b * largest and (off[row >= 2.0 ** -a * largest] == 0).all()
