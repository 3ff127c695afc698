"""mx_block_gemm_grouped_k_rows on the host: its refusals are those of the call without rows, and a number of rows
that is none."""
import pytest

from test_grouped_cpu import A, BS, E, INVALID, L, OK, P, UNSUPPORTED, Y, cols_args  # noqa: F401 (L is a fixture)


def args(**k):
    a = cols_args(**k)
    return a[:12] + [k.get("rows", 300)] + a[12:]


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=-1 << 40), dict(M=-1), dict(cols=895), dict(groups=-1), dict(lda=895),
                                 dict(ldsb=259), dict(ldc=259), dict(ldcg=70 * 260 - 1), dict(ends=None), dict(c=None), dict(c=A),
                                 dict(c=BS), dict(c=E), dict(a=P(Y.value + 4 * 5 * 70 * 260 - 1))], ids=str)
def test_rejects(L, bad):
    assert L.mx_block_gemm_grouped_k_rows(*args(**bad)) == INVALID


@pytest.mark.parametrize("bad", [dict(rows=1 << 31), dict(rows=1 << 62), dict(groups=(1 << 16) + 1)], ids=str)
def test_limits(L, bad):
    assert L.mx_block_gemm_grouped_k_rows(*args(**bad)) == UNSUPPORTED


def test_empty_calls(L):
    none = dict(a=None, as_=None, b=None, bs=None, ends=None, c=None)
    for k in (dict(M=0), dict(N=0), dict(groups=0), dict(M=0, rows=0, cols=0)):
        assert L.mx_block_gemm_grouped_k_rows(*args(**k, **none)) == OK
