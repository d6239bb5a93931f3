"""Host-side rules of the operators at the ends of a language model."""
from test_host_rules import run


def test_chunks_read_the_places_that_there_are(tmp_path):
    run("embed_chunks_test", tmp_path)


def test_copied_rows_keep_the_threads_busy(tmp_path):
    run("pack_shape_test", tmp_path)
