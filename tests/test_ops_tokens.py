"""How gemm_int8 takes bf16 tokens, without a GPU: made to integers inside the product for a few tokens of few columns,
by a launch before it otherwise (calls of the library are noted, none is made)."""
import types

import pytest

import sparse_mask_search_amd as sms

torch = pytest.importorskip("torch")


@pytest.fixture()
def launches(monkeypatch):
    from sparse_mask_search_amd import _ops
    names = []
    monkeypatch.setattr(_ops, "_matrix", lambda *a: None)
    monkeypatch.setattr(_ops, "_run", lambda torch, where, device, fn, *args: names.append((where, *args)))
    monkeypatch.setattr(_ops, "lib", lambda: types.SimpleNamespace(tsenor_quant_int8=None, tsenor_gemm_int8=None))
    return names


@pytest.mark.parametrize("rows,m,k,dtype,inside", [
    (1, 4096, 4096, "bfloat16", True), (1, 32000, 4096, "bfloat16", True), (1, 100000, 32768, "bfloat16", True),
    (1, 64, 32769, "bfloat16", False), (4, 8192, 4096, "bfloat16", True), (8, 4096, 4096, "bfloat16", True),
    (8, 512, 4097, "bfloat16", False), (2, 11008, 4096, "bfloat16", True), (3, 11008, 4096, "bfloat16", False),
    (2, 32000, 4096, "bfloat16", False), (9, 512, 512, "bfloat16", False), (16, 4096, 2048, "bfloat16", False),
    (17, 64, 128, "bfloat16", False), (1, 64, 128, "float32", False),
])
def test_where_tokens_become_integers(launches, rows, m, k, dtype, inside):
    x = torch.empty(rows, k, dtype=getattr(torch, dtype))
    a = sms.DenseInt8(torch.empty(m, -(-k // 128) * 128, dtype=torch.int8), torch.empty(m), k)
    y = sms.gemm_int8.__wrapped__(torch, x, a)
    assert y.shape == (rows, m)
    gemm = launches[-1]
    assert [c[0] for c in launches] == (["tsenor_gemm_int8"] if inside else ["tsenor_quant_int8", "tsenor_gemm_int8"])
    assert gemm[2] == (1 if inside else 3) and (gemm[3] is None) == inside and gemm[4] == rows
