"""What kd_policy_loss refuses before it looks at a tensor's place or type: meanings
that cannot be told from sizes, and options that would have no effect. (The tensors
are on the CPU: a call that passes these checks is refused for that.)"""
import pytest
import torch

from lm_head_top_gb300 import kdkl

T = 6
X = torch.zeros(T)


def _cu(S):
    return torch.tensor([0] + [T] * S, dtype=torch.int32)


def _refused(match, *a, **kw):
    with pytest.raises(ValueError, match=match):
        kdkl.kd_policy_loss(*a, **kw)


def test_as_many_sequences_as_tokens_need_the_word():
    """Advantages of T = S values: one a token, or one a sequence, some of them empty."""
    _refused("advantage_per_sequence", X, None, None, X, None, _cu(T))
    _refused("advantage_per_sequence", X, None, None, X, None, _cu(T), reduction="sequence")
    for word in (True, False):
        _refused("CUDA", X, None, None, X, None, _cu(T), advantage_per_sequence=word)


@pytest.mark.parametrize("n,word", [(2, False), (T, True), (3, True), (3, False)])
def test_the_word_has_to_fit_the_size(n, word):
    _refused("advantages", X, None, None, torch.zeros(n), None, _cu(2), advantage_per_sequence=word)


def test_per_sequence_needs_sequences():
    _refused("cu_seqlens", X, None, None, X, advantage_per_sequence=True)


def test_sizes_that_differ_need_no_word():
    _refused("CUDA", X, None, None, torch.zeros(2), None, _cu(2))
    _refused("CUDA", X, None, None, X, None, _cu(2))
    _refused("CUDA", X, None, None, X)


def test_one_sequence_of_one_token_needs_no_word():
    one = torch.zeros(1)
    _refused("CUDA", one, None, None, one, None, torch.tensor([0, 1], dtype=torch.int32))


@pytest.mark.parametrize("kl_coef", [0.1, -0.1])
def test_a_kl_term_needs_its_reference(kl_coef):
    _refused("ref_logp", X, X, None, X, kl_coef=kl_coef)
    _refused("CUDA", X, X, None, X, kl_coef=0.0)
    _refused("CUDA", X, X, X, X, kl_coef=kl_coef)
