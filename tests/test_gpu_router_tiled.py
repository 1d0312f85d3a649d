"""det_router_balance with many tokens or many slots and few experts: calls of few
logits that still take several workgroups per segment."""
import pytest

from tests.test_gpu_router_balance import BF, F32, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,dtype,offs", [(65536, 2, 2, BF, [0, 65536]), (16384, 8, 8, F32, [0, 16384]),
                                              (16384, 8, 8, BF, [5, 3000, 3000, 16000]), (40000, 1, 1, F32, [0, 7, 40000]),
                                              (9000, 9, 4, BF, [0, 9000]), (220, 4, 3001, F32, [0, 100, 219]),
                                              (1, 2, 65536, F32, [0, 1])])
def test_many_tokens_or_slots_and_few_experts(T, E, K, dtype, offs, score):
    check(T, E, K, dtype, offs, score, seed=T + K)
