"""The look at the kernels' error words that follows every GPU test file, with
the words faked."""
import pytest

from waits import assert_none_gave_up


class Fake:
    def __init__(self, block=(0, 0), quant=(0, 0, 0)):
        self.block, self.quant, self.cleared = block, quant, 0

    def block_device_errors(self, clear=False):
        self.cleared += clear
        return self.block

    def glu_quant_device_errors(self, clear=False):
        self.cleared += clear
        return self.quant


def test_clean_words_pass_and_are_cleared():
    f = Fake()
    assert_none_gave_up(f, "here")
    assert f.cleared == 2


@pytest.mark.parametrize("words", [dict(block=(0, 1)), dict(block=(-4, 0)), dict(quant=(0, 4, 0)), dict(quant=(0, 0, 2)), dict(quant=(-4, 0, 0))])
def test_a_mark_or_an_unreadable_word_fails(words):
    f = Fake(**words)
    with pytest.raises(AssertionError, match="waits gave up in here"):
        assert_none_gave_up(f, "here")
    assert f.cleared == 2


def test_every_gpu_file_is_looked_at(request):
    """The fixture that does it is in use for every file."""
    assert "no_wait_gave_up" in request.fixturenames
