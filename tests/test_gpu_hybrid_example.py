"""The example of the softmax-attention layer: the operators together, as a serving and a training program use them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_17_gb300 import build

    build.build()


def test_tree_rows_equal_decoding_one_by_one():
    from examples.hybrid_attention import verify_a_tree

    # the same tokens and keys: what differs are the bf16 roundings of the weights and of the rows, 2^-8 each on
    # either side
    assert verify_a_tree() <= 4 * 2.0 ** -8


def test_a_deep_and_a_wide_tree():
    from examples.hybrid_attention import verify_a_tree

    chain = tuple(range(-1, 39))
    assert verify_a_tree(prompt=(33, 200), parents=chain, accepted=(0, 1, 2, 3)) <= 4 * 2.0 ** -8
    wide = (-1,) * 70  # more than one mask word
    assert verify_a_tree(prompt=(5, 1), parents=wide, accepted=(69,)) <= 4 * 2.0 ** -8


def test_a_step_on_the_norms_weights_lowers_the_loss():
    from examples.hybrid_attention import train_the_norm

    before, after = train_the_norm()
    assert after < before
