"""Inputs of attention whose results count keys (or queries), so that one too
few or too many shows at any length.

With q = 0 all scores are 0: every weight is 1, its sum the number of keys that
a query sees, all exact.  Columns of v (dout, k or q in the gradients) mark the
rows: row j has a 1 in column j mod M less an offset, if that is one, with M so
large that a column's count stays small beside the steps of bf16.
"""

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24
MOST = 60  # marked rows of a column


def period(rows, dim):
    """M for sequences of up to `rows` marked rows: a multiple of dim."""
    return dim * max(1, -(-rows // (MOST * dim)))


def marks(index, dim, m, offset, dtype=torch.bfloat16):
    """[rows, dim]: the marks of rows with these indices in their sequence."""
    col = torch.arange(dim, device=index.device) + offset
    return (index[:, None] % m == col).to(dtype)


def below(limit, dim, m, offset):
    """[.., dim]: marked rows of each column among the first `limit` of a sequence."""
    col = torch.arange(dim, device=limit.device) + offset
    return torch.clamp((limit[..., None] - col + m - 1) // m, min=0)


def check_mean(out, lse, limit, dim, m, offset):
    """The forward call's results of rows that see `limit` keys."""
    count = below(limit, dim, m, offset).double()
    keys = limit.double()
    want = torch.where(limit[..., None] > 0, count / keys[..., None], torch.zeros_like(count))
    # 1 / sum, its product with each of at most 152 parts and their sum, then bf16
    err = (out.double() - want).abs()
    assert (err <= (U16 + 160 * U32) * want).all(), "keys counted in out"
    # log2 (an ulp, twice U32), its factor and their product
    log = torch.log(keys)
    assert ((lse.double() - log).abs() <= 4 * U32 * log)[limit > 0].all(), "keys counted in lse"
    assert (lse[limit <= 0] == -float("inf")).all()
