"""Workspace sizes of the K8/V8 attention calls: none for head counts that the
calls refuse, one that the call takes for the others.  (Without a GPU every size
is 0.)"""
import pytest
import torch

from cases import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from fp8_paged_kv_append_gb300 import k16v8
    k16v8.load_library()
    return k16v8


def decode(K, hq, hkv, ws_bytes):
    """Status of a decode call of one sequence without positions."""
    cache = [torch.zeros((1, hkv, 16, 128), dtype=torch.uint8, device=dev()) for _ in range(2)]
    cache.append(torch.ones((1, hkv, 2), device=dev()))
    q = torch.zeros((1, hq, 128), dtype=torch.float16, device=dev())
    try:
        K.k16v8_paged_decode_attention_k8v8(
            q, *cache, torch.zeros((1, 1), dtype=torch.int32, device=dev()),
            torch.zeros(1, dtype=torch.int32, device=dev()), 1.0,
            torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev()), q)
    except K.K16V8Error as e:
        return e.status
    return K.K16V8_OK


@pytest.mark.parametrize("hq", [1, 2, 3, 5, 6, 9, 41])
def test_no_size_where_decode_refuses_the_heads(K, hq):
    assert K.k16v8_decode_workspace_size_k8v8(1, hq, 128) == 0
    for hkv in (1, max(1, hq // 4)):
        assert decode(K, hq, hkv, 1 << 24) != K.K16V8_OK
        assert K.k16v8_attention_workspace_size_k8v8(8, hq, hkv, 128) == 0


@pytest.mark.parametrize("hkv", [1, 2, 10])
def test_the_size_is_enough(K, hkv):
    n = K.k16v8_decode_workspace_size_k8v8(1, 4 * hkv, 128)
    assert n > 0 and decode(K, 4 * hkv, hkv, n) == K.K16V8_OK
    assert decode(K, 4 * hkv, hkv, n - 1) != K.K16V8_OK
