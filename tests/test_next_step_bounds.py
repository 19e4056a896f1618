"""The next step's tables on the GPU where the free stack has nearly 2^31 places."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


@pytest.fixture(scope="module")
def stack():
    x = torch.full(((1 << 31) - 1,), 77, dtype=torch.int32, device=DEV)
    yield x
    del x
    torch.cuda.empty_cache()


def pool(stack, n_free):
    from speculative_decoding_block_ingest_gb300 import target
    table = i32([[3, 4, 5], [6, 8, -1]])
    return target, target.PagePool(stack, i32([n_free]), table, i32([40, 20]), i32([0, 1, 2]), page_size=16)


def test_pages_given_to_a_stack_that_says_it_is_full(stack):
    """The height is bounded to the stack's places, and nothing is written behind or before them."""
    n = stack.shape[0]
    for n_free, kept in ((n, n), (n - 2, n), (n - 5, n)):
        stack[-8:] = 77
        T, p = pool(stack, n_free)
        T.next_step(p, i32([0, 0]), n_rows=4, keep=i32([0, 0]))        # all five pages
        assert p.n_free.tolist() == [kept] and p.kv_len.tolist() == [0, 0]
        want = {n: [], n - 2: [8, 6], n - 5: [8, 6, 5, 4, 3]}[n_free]
        assert stack[-8:].tolist() == [77] * (8 - (n - n_free)) + want
        assert stack[:8].tolist() == [77] * 8


def test_pages_taken_from_its_top(stack):
    n = stack.shape[0]
    stack[-4:] = i32([90, 91, 92, 93])
    T, p = pool(stack, n)
    slots = torch.full((10,), -1, dtype=torch.int64, device=DEV)
    T.next_step(p, i32([0, 10]), slots=slots, keep=i32([17, -1]))       # one page given, none needed
    assert p.n_free.tolist() == [n] and slots.tolist() == [8 * 16 + 4 + i for i in range(10)]
    stack[-4:] = i32([90, 91, 92, 93])
    T, p = pool(stack, n)
    T.next_step(p, i32([0, 28]), n_rows=30)                              # a page needed
    assert p.n_free.tolist() == [n - 1] and p.block_table.tolist() == [[3, 4, 5], [6, 8, 93]]
