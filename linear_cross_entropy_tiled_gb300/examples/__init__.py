"""Small runnable uses of the package."""
