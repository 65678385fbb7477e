"""pa_bm_evict where nothing, or not everything, can be cut."""
import pytest


@pytest.fixture(scope="module")
def manager():
    from paged_kv_cache_390_b200 import build
    from paged_kv_cache_390_b200.block_manager import BlockManager
    build.build()
    return lambda n=20, bs=4: BlockManager(n, bs, 4, True)


@pytest.mark.parametrize("tokens,keep", [(6, 6), (6, 50), (8, 8), (3, 4)])
def test_a_sequence_that_keeps_everything_goes_on_in_the_prefix_cache(manager, tokens, keep):
    """It is moved whole, so the blocks that it fills later hold its tokens one to one and
    are found by other sequences."""
    m = manager()
    text = list(range(100, 116))
    m.add_sequence(1, text[:tokens])
    m.evict([1], keep)
    for t in text[tokens:]:
        m.append_token(1, t)
    blocks, n = m.block_table(1)
    assert n == 16
    _, cached = m.add_sequence(2, text + [7])
    assert cached == 16
    # the blocks filled after the move are the first sequence's own
    first = tokens // 4
    assert m.block_table(2)[0].tolist()[first:4] == blocks.tolist()[first:4]
    for s in (1, 2):
        m.free_sequence(s)
    assert m.free_gpu_blocks == 20


def test_a_cut_sequence_stays_out_of_the_prefix_cache(manager):
    m = manager()
    text = list(range(100, 116))
    m.add_sequence(1, text[:6])
    m.evict([1], 5)                                        # one token fewer: cut
    m.evict([1], 50)                                       # whole again, but still cut
    for t in text[6:]:
        m.append_token(1, t)
    _, cached = m.add_sequence(2, text + [7])
    assert cached == 4                                     # the prompt's own first block


def test_a_nearly_full_pool_is_cut_sequence_by_sequence(manager):
    from paged_kv_cache_390_b200 import pa
    m = manager(n=18)
    for s in range(4):
        m.add_sequence(s, range(100 * s, 100 * s + 16))    # four blocks each, two free
    with pytest.raises(pa.PAError) as e:
        m.evict([0, 1, 2, 3], 8)                           # eight fresh ones at once
    assert e.value.status == pa.PA_ERR_NO_SPACE
    assert [m.block_table(s)[1] for s in range(4)] == [16] * 4 and m.free_gpu_blocks == 2
    for s in range(4):
        assert m.evict([s], 8).shape == (1, 2)
    assert m.free_gpu_blocks == 10
