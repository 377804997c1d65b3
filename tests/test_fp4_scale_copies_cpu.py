"""The bulk copies of activations' scale bytes (8 a row): their sources, sizes and readers, taken from
the kernels' source and evaluated for rows of either parity (CPU). A copy starts on a 16-byte
boundary, is a whole number of 16 bytes, stays inside the buffer of an even number of rows, and a
row's scales are read from where its copy put them."""
import re
from types import SimpleNamespace

import pytest

from test_fp4_source_cpu import arguments, code


def value(expr, **names):
    """A C expression of integers: casts dropped, one conditional at its top allowed."""
    expr = re.sub(r"\((?:size_t|int|long long|uint32_t)\)", "", expr).replace("1ll", "1")
    m = re.fullmatch(r"\s*(.+?) \? (.+?) : (.+)", expr, flags=re.S)
    if m:
        return value(m[2] if value(m[1], **names) else m[3], **names)
    return int(eval(" ".join(expr.split()), {"min": min}, names))


def define(text, name):
    return re.search(r"\b%s = ([^;,]+)[;,]" % name, text)[1]


def bulk(text, first):
    """Arguments of the copy whose destination is `first`."""
    found = []
    for m in re.finditer(r"\bbulk_load\(", text):
        args = [a.strip() for a in re.split(r",(?![^(]*\))", arguments(text, m.end()))]
        if args[0] == first:
            found.append(args)
    assert len(found) == 1
    return found[0]


def few_rows(text):
    """(source byte of stage kt, bytes, byte read for the tile's row i) of rows_fp4.cu."""
    at = re.search(r"sx = \(G == kFc1 \? p\.xs : p\.hs\) \+ ([^;]+);", text)[1]
    src, size = bulk(text, "s + kSxAt")[1:3]
    assert src.startswith("sx + ") and size == "sbx" and "np = scale_rows(p.N)" in text
    read = re.search(r"s \+ kSxAt \+ (\(.+?\) \* 8)\)", text)[1]

    def of(row, rows, np_, kt):
        t = SimpleNamespace(row=row, rows=rows)
        sr = value(define(text, "sr"), t=t)
        start = value(at, sr=sr) + value(src[len("sx + "):], kt=kt, np=np_)
        odd = value(define(text, "odd"), t=t)
        return start, value(define(text, "sbx"), t=t), lambda i: value(read, odd=odd, lane=i)

    return of, 32


def many_rows(text):
    """The same of grouped_gemm_fp4.cu."""
    at = re.search(r"sa = \(MODE == FC1 \? p\.xs : p\.hs\) \+ ([^;]+);", text)[1]
    src, size = bulk(text, "s")[1:3]
    assert src.startswith("sa + ") and size == "ba" and "np = scale_rows(p.N)" in text
    assert define(text, "ba") == "n == t.n0 ? rows : 0"
    read = re.search(r"s \+ (\(odd \+ .+?\) \* 8)\)", text)[1]

    def of(row, rows, np_, kt):
        t = SimpleNamespace(row0=row // 2, m0=row - row // 2, rows=rows)
        r0 = value(define(text, "r0"), row=row)
        start = value(at, r0=r0) + value(src[len("sa + "):], kt=kt, np=np_)
        odd = value(define(text, "odd"), t=t)
        return (start, value(define(text, "uint32_t rows"), t=t, row=row),
                lambda i: value(read, odd=odd, i=i // 32, lane=i % 32))

    return of, 128


def check(text, which):
    of, most = which(text)
    for N in (1, 2, 3, 33, 130, 131, 257):
        np_ = (N + 1) & ~1
        for row in {0, 1, 2, 3, N // 2, N - 1} & set(range(N)):
            for rows in {1, 2, 3, 31, most, N - row} & set(range(1, min(most, N - row) + 1)):
                for kt in (0, 3):
                    start, size, read = of(row, rows, np_, kt)
                    assert start % 16 == 0 and size % 16 == 0 and size > 0
                    assert kt * np_ * 8 <= start and start + size <= (kt + 1) * np_ * 8
                    for i in (0, rows - 1):
                        assert start + read(i) == (kt * np_ + row + i) * 8 and read(i) + 8 <= size


CASES = [("rows_fp4.cu", few_rows), ("grouped_gemm_fp4.cu", many_rows)]


@pytest.mark.parametrize("name,which", CASES)
def test_copies_of_scales(name, which):
    check(code(name), which)
    assert "(n + 1) & ~1ll" in code("fp4_mma.cuh")  # scale_rows


def test_no_rows_no_copy():
    text = code("grouped_gemm_fp4.cu")
    assert value(define(text, "uint32_t rows"), t=SimpleNamespace(rows=0), row=5) == 0
    assert re.search(r"if \(ba\) bulk_load\(s, ", text)


@pytest.mark.parametrize("name,which,there,planted", [
    ("rows_fp4.cu", few_rows, "sr = t.row & ~1ll", "sr = t.row"),
    ("rows_fp4.cu", few_rows, "t.rows + 1) & ~1) * 8", "t.rows) & ~1) * 8"),
    ("rows_fp4.cu", few_rows, "(odd + lane) * 8", "(lane) * 8"),
    ("rows_fp4.cu", few_rows, "odd = (int)(t.row & 1)", "odd = 0"),
    ("grouped_gemm_fp4.cu", many_rows, "r0 = row & ~1ll", "r0 = row"),
    ("grouped_gemm_fp4.cu", many_rows, "t.rows + 1) & ~1) * 8", "t.rows + 2) & ~1) * 8"),
    ("grouped_gemm_fp4.cu", many_rows, "odd = (t.row0 + t.m0) & 1", "odd = t.m0 & 1"),
    ("grouped_gemm_fp4.cu", many_rows, "(odd + 32 * i + lane) * 8", "(odd + 16 * i + lane) * 8"),
])
def test_the_check_sees_planted_mistakes(name, which, there, planted):
    text = code(name)
    assert there in text
    with pytest.raises(AssertionError):
        check(text.replace(there, planted), which)
